"""Host-side checks of include/muon_lm.h and its binding (no GPU needed): the
library exports what the header declares, bad arguments give the documented
status before a device is touched, and the binding refuses what it cannot pass
on."""
import ctypes
import os
import re

import pytest
import torch

import newton_schulz_07_gb300 as ns
from newton_schulz_07_gb300 import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 4096
BAD, ALIGN, WS = _lib.ERR_INVALID_ARG, _lib.ERR_ALIGNMENT, _lib.ERR_WORKSPACE


def test_library_exports_every_declared_function():
    text = open(os.path.join(ROOT, "include", "muon_lm.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    declared = set(re.findall(r"\b(muon_\w+)\s*\(", text))
    assert declared == set(_lib.LM_SIGNATURES)
    assert all(hasattr(_lib.lib(), n) for n in declared)
    assert all(hasattr(ns, n) for n in declared if not n.endswith("_workspace_size"))


def test_header_compiles_as_c_and_cpp(tmp_path):
    import shutil
    import subprocess

    cuda_inc = "/usr/local/cuda/include"
    cc, cxx = shutil.which("gcc"), shutil.which("g++")
    if not (cc and cxx and os.path.exists(os.path.join(cuda_inc, "cuda_runtime_api.h"))):
        pytest.skip("no host C compiler or CUDA headers")
    src = tmp_path / "use_header.c"
    src.write_text('#include "muon_lm.h"\nint main(void) { size_t n = 0; return '
                   "muon_embed_grad_workspace_size(1, 8, 8, &n) + MUON_LM_F32; }\n")
    inc = ["-I" + os.path.join(ROOT, "include"), "-I" + cuda_inc]
    for cmd in ([cc, "-std=c99"], [cxx, "-std=c++17", "-x", "c++"]):
        p = subprocess.run(cmd + ["-Wall", "-Werror", "-fsyntax-only"] + inc + [str(src)], stdout=subprocess.PIPE,
                           stderr=subprocess.STDOUT, text=True)
        assert p.returncode == 0, p.stdout


def _embed(**kw):
    a = dict(table=P, tt=0, vocab=10, dim=8, ids=P, bits=32, tokens=4, scale=1.0, out=1 << 20, ot=0)
    a.update(kw)
    return _lib.lib().muon_embed(a["table"], a["tt"], a["vocab"], a["dim"], a["ids"], a["bits"], a["tokens"],
                                 a["scale"], a["out"], a["ot"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=-1), BAD), (dict(vocab=-1), BAD), (dict(dim=-1), BAD), (dict(tokens=(1 << 30) + 1), BAD),
    (dict(dim=(1 << 20) + 1), BAD), (dict(bits=16), BAD), (dict(tt=2), BAD), (dict(ot=-1), BAD),
    (dict(scale=float("nan")), BAD), (dict(scale=float("inf")), BAD), (dict(table=None), BAD), (dict(ids=None), BAD),
    (dict(out=None), BAD), (dict(out=P), BAD), (dict(table=P + 1), ALIGN), (dict(ot=1, out=(1 << 20) + 2), ALIGN),
    (dict(ids=P + 2), ALIGN), (dict(ids=P + 4, bits=64), ALIGN), (dict(tokens=0, out=None), 0),
    (dict(dim=0, table=None, out=None), 0)])
def test_embed_refusals(kw, code):
    assert _embed(**kw) == code


def _embed_grad(**kw):
    a = dict(dy=1 << 20, dt=0, ids=P, bits=32, tokens=1600, vocab=10, dim=8, scale=1.0, out=1 << 21, ot=1, acc=0, ws=1 << 22,
             wsb=1 << 20)
    a.update(kw)
    return _lib.lib().muon_embed_grad(a["dy"], a["dt"], a["ids"], a["bits"], a["tokens"], a["vocab"], a["dim"], a["scale"],
                                      a["out"], a["ot"], a["acc"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=-1), BAD), (dict(vocab=(1 << 30) + 1), BAD), (dict(bits=8), BAD), (dict(dt=3), BAD), (dict(ot=3), BAD),
    (dict(scale=float("nan")), BAD), (dict(dy=None), BAD), (dict(ids=None), BAD), (dict(out=None), BAD),
    (dict(out=1 << 20), BAD), (dict(dy=(1 << 20) + 1), ALIGN), (dict(out=(1 << 21) + 2), ALIGN),
    (dict(ws=(1 << 22) + 16), ALIGN), (dict(ws=None), WS), (dict(wsb=64), WS), (dict(vocab=0, out=None), 0),
    (dict(dim=0, out=None), 0)])
def test_embed_grad_refusals(kw, code):
    assert _embed_grad(**kw) == code


def _norm(**kw):
    a = dict(x=P, xt=0, w=P, b=P, wt=1, rows=3, dim=8, eps=1e-5, y=P, mean=P, rstd=P)
    a.update(kw)
    return _lib.lib().muon_layer_norm(a["x"], a["xt"], a["w"], a["b"], a["wt"], a["rows"], a["dim"], a["eps"], a["y"],
                                      a["mean"], a["rstd"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), BAD), (dict(dim=0), BAD), (dict(dim=(1 << 20) + 1), BAD), (dict(rows=(1 << 30) + 1), BAD),
    (dict(xt=2), BAD), (dict(wt=2), BAD), (dict(eps=-1.0), BAD), (dict(eps=float("nan")), BAD), (dict(x=None), BAD),
    (dict(w=None), BAD), (dict(y=None), BAD), (dict(x=P + 1), ALIGN), (dict(y=P + 1), ALIGN), (dict(w=P + 2), ALIGN),
    (dict(b=P + 2), ALIGN), (dict(mean=P + 2), ALIGN), (dict(rows=0, x=None, y=None), 0)])
def test_layer_norm_refusals(kw, code):
    assert _norm(**kw) == code


def _norm_grad(**kw):
    a = dict(dy=P, x=P, xt=0, w=P, wt=1, mean=P, rstd=P, rows=30000, dim=8, dx=P, dw=P, db=P, ws=P, wsb=1 << 20)
    a.update(kw)
    return _lib.lib().muon_layer_norm_grad(a["dy"], a["x"], a["xt"], a["w"], a["wt"], a["mean"], a["rstd"], a["rows"],
                                           a["dim"], a["dx"], a["dw"], a["db"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), BAD), (dict(dim=0), BAD), (dict(xt=2), BAD), (dict(wt=-1), BAD), (dict(dy=None), BAD),
    (dict(x=None), BAD), (dict(w=None), BAD), (dict(mean=None), BAD), (dict(rstd=None), BAD), (dict(dx=None), BAD),
    (dict(dw=None), BAD), (dict(dx=P + 1), ALIGN), (dict(db=P + 2), ALIGN), (dict(ws=P + 16), ALIGN),
    (dict(ws=None), WS), (dict(wsb=16), WS), (dict(rows=0, dim=0, dw=None), 0)])
def test_layer_norm_grad_refusals(kw, code):
    assert _norm_grad(**kw) == code


H, W, T, L, DH, DW, SP = (i << 24 for i in range(1, 8))
BIG = 1 << 40


def _head(**kw):
    a = dict(h=H, w=W, n=5, v=100, d=16, t=T, bits=64, ignore=-100, loss=L, ws=SP, wsb=BIG)
    a.update(kw)
    return _lib.lib().muon_head_loss(a["h"], a["w"], a["n"], a["v"], a["d"], a["t"], a["bits"], a["ignore"], a["loss"],
                                     a["ws"], a["wsb"], None)


HEAD = [(dict(n=-1), BAD), (dict(v=-1), BAD), (dict(d=0), BAD), (dict(d=-8), BAD), (dict(d=12), ALIGN),
        (dict(n=(1 << 30) + 1), BAD), (dict(v=(1 << 30) + 1), BAD), (dict(d=(1 << 20) + 8), BAD), (dict(bits=16), BAD),
        (dict(h=None), BAD), (dict(w=None), BAD), (dict(t=None), BAD), (dict(loss=None), BAD), (dict(h=H + 8), ALIGN),
        (dict(w=W + 2), ALIGN), (dict(t=T + 4), ALIGN), (dict(loss=L + 2), ALIGN), (dict(ws=SP + 128), ALIGN),
        (dict(ws=None), WS), (dict(wsb=1000), WS)]


@pytest.mark.parametrize("kw,code", HEAD + [(dict(n=0, h=None, loss=None, ws=None), 0)])
def test_head_loss_refusals(kw, code):
    assert _head(**kw) == code


def _head_grad(**kw):
    a = dict(h=H, w=W, n=5, v=100, d=16, t=T, bits=64, ignore=-100, dloss=None, pieces=0, loss=L, dh=DH, dw=DW, dt=0, acc=0,
             ws=SP, wsb=BIG)
    a.update(kw)
    return _lib.lib().muon_head_loss_grad(a["h"], a["w"], a["n"], a["v"], a["d"], a["t"], a["bits"], a["ignore"], a["dloss"],
                                          a["pieces"], a["loss"], a["dh"], a["dw"], a["dt"], a["acc"], a["ws"], a["wsb"],
                                          None)


@pytest.mark.parametrize("kw,code", HEAD + [
    (dict(pieces=-1), BAD), (dict(dt=2), BAD), (dict(acc=1), BAD), (dict(dh=None), BAD), (dict(dw=None), BAD),
    (dict(dh=H), BAD), (dict(dh=W), BAD), (dict(dw=H), BAD), (dict(dw=W + 16), BAD), (dict(dw=DH + 32), BAD),
    (dict(dh=DH + 8), ALIGN), (dict(dw=DW + 4), ALIGN), (dict(dloss=L + 2), ALIGN),
    (dict(n=0, v=0, h=None, w=None, t=None, loss=None, dh=None, dw=None, ws=None), _lib.ERR_UNSUPPORTED_DEVICE
     if not torch.cuda.is_available() else 0)])
def test_head_loss_grad_refusals(kw, code):
    assert _head_grad(**kw) == code


def test_head_workspace():
    size = ns.head_workspace_size
    # One piece holds tokens x vocab in bf16; more pieces hold less; the losses
    # alone hold none of it.
    assert size(1000, 50000, 64, True, 1) >= 2 * 1000 * 50000 > size(1000, 50000, 64, True, 8) > size(1000, 50000, 64, False)
    # By default a piece is at most about 4 GiB.
    assert 1 << 32 <= size(200000, 131072, 64) < 6 << 30
    assert size(0, 50000, 64) == size(1000, 0, 64) == 0
    for bad in ((-1, 10, 8), (1, 10, 12), (1, 10, 0)):
        with pytest.raises(ns.MuonNSError):
            size(*bad)
    with pytest.raises(ns.MuonNSError):
        size(1, 10, 8, True, -1)


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device path")
def test_valid_calls_without_a_device_are_unsupported():
    for call in (_embed, _embed_grad, _norm, _norm_grad, _head, _head_grad):
        assert call() == _lib.ERR_UNSUPPORTED_DEVICE


def test_workspace_sizes():
    assert ns.embed_grad_workspace_size(0, 10, 8) == 0 and ns.layer_norm_grad_workspace_size(0, 8) == 0
    # Sorted pairs twice, two partial rows a piece of 32 positions.
    assert ns.embed_grad_workspace_size(2000, 100, 64) >= 16 * 2000 + 32 * 2 * 64 * 4
    assert ns.layer_norm_grad_workspace_size(50000, 24) >= 2 * 24 * 4
    # Few tokens and few rows need none.
    assert ns.embed_grad_workspace_size(256, 100, 64) == 0 < ns.embed_grad_workspace_size(257, 100, 64)
    assert ns.layer_norm_grad_workspace_size(7, 4096) == 0
    with pytest.raises(ns.MuonNSError):
        ns.embed_grad_workspace_size(-1, 10, 8)
    with pytest.raises(ns.MuonNSError):
        ns.layer_norm_grad_workspace_size(4, 0)
    assert _lib.lib().muon_embed_grad_workspace_size(1, 1, 1, None) == BAD
    assert _lib.lib().muon_layer_norm_grad_workspace_size(1, 1, ctypes.POINTER(ctypes.c_size_t)()) == BAD


def test_binding_refuses_host_tensors():
    x, ids = torch.ones(4, 8), torch.zeros(4, dtype=torch.int64)
    for f in (lambda: ns.muon_embed(x, ids), lambda: ns.muon_embed_grad(x, ids, 10), lambda: ns.muon_layer_norm(x, x[0]),
              lambda: ns.muon_layer_norm_grad(x, x, x[0], x[:, 0], x[:, 0]),
              lambda: ns.muon_head_loss(x.bfloat16(), x.bfloat16(), ids),
              lambda: ns.muon_head_loss_grad(x.bfloat16(), x.bfloat16(), ids)):
        with pytest.raises(TypeError):
            f()


@pytest.mark.parametrize("size", [lambda d: ns.embed_grad_workspace_size(2000, 100, d), lambda d: ns.layer_norm_grad_workspace_size(50000, d),
                                  lambda d: ns.head_workspace_size(1000, 500, d), lambda d: ns.head_workspace_size(1000, 500, 64, True, d)])
def test_sizes_past_an_int_are_refused(size):
    # A C int would keep the low 32 bits: 64 of 2^32 + 64.
    for n in ((1 << 32) + 64, (1 << 31) + 64, -(1 << 32) + 64):
        with pytest.raises(ns.MuonNSError) as e:
            size(n)
        assert e.value.status == BAD
    assert size(64) > 0


@pytest.mark.parametrize("call", [_embed_grad, _norm_grad, _head, _head_grad])
def test_a_workspace_that_is_not_needed_is_not_looked_at(call):
    # Past the checks of arguments: done, or the lack of a device.
    few = {_embed_grad: dict(tokens=0, acc=1), _norm_grad: dict(rows=0, dim=0), _head: dict(n=0),
           _head_grad: dict(n=0, v=0, dw=None)}[call]
    for ws in (None, SP + 16):
        assert call(ws=ws, wsb=16, **few) in (0, _lib.ERR_UNSUPPORTED_DEVICE)
    if call in (_embed_grad, _norm_grad) and not torch.cuda.is_available():
        few = dict(tokens=256) if call is _embed_grad else dict(rows=3)
        assert call(ws=SP + 16, wsb=0, **few) == _lib.ERR_UNSUPPORTED_DEVICE
