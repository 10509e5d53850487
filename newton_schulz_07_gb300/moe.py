"""Binding of include/muon_moe.h: the operators of a block with experts.

As in lm.py, argument marshalling only; names follow the C entry points.
Tensors are contiguous CUDA tensors on one device, work is enqueued on that
device's current stream, and autograd is not involved: the backward pass is the
caller's to call.
"""
from __future__ import annotations

import torch

from . import _lib
from .lm import _BF16, _F32, _TYPES, _call, _int, _shaped, _size, _tensor, _workspace

_I32 = {torch.int32: 0}
_E4M3 = {torch.float8_e4m3fn: 0}
BLOCK = 128  # values that share a scale in 8-bit storage


def _blocks(n):
    return -(-n // BLOCK)


def _error(t, device):
    """Pointer of an optional int32 device word."""
    if t is None:
        return None
    _tensor(t, "error", _I32, device)
    if t.numel() < 1:
        raise ValueError("error must hold an int32")
    return t.data_ptr()


def _out(t, shape, dtype, like, name):
    """t checked, or a new tensor of that shape and dtype where `like` is."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    _tensor(t, name, {dtype: 0}, like.get_device())
    _shaped(t, shape, name)
    return t


# ---------------------------------------------------------------- RMS norm --

def _norm_args(x, weight, residual):
    """(device, x's type code, weight's, shape, rows, dim, residual's pointer)."""
    xt = _tensor(x, "x")
    dev = x.get_device()
    wt = _tensor(weight, "weight", device=dev)
    shape = x.shape
    if not shape:
        raise ValueError("x must have an axis to normalise over")
    dim = _int(shape[-1], "dim")
    _shaped(weight, (dim,), "weight")
    rp = None
    if residual is not None:
        if _tensor(residual, "residual", device=dev) != xt:
            raise TypeError("residual must have x's dtype")
        _shaped(residual, shape, "residual")
        rp = residual.data_ptr()
    return dev, xt, wt, shape, dim, rp


def muon_rms_norm(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None, eps: float = 1e-6,
                  out: torch.Tensor | None = None, total: torch.Tensor | None = None):
    """Root-mean-square norm over the last axis of x + residual.  Returns (y, s,
    rstd): y and the sum s (x itself without a residual) of x's shape and dtype,
    rstd fp32 of x's shape without its last axis.  weight: bfloat16 or float32.
    `out` (y) and `total` (s) may each be x or the residual.  Written over x without
    a residual, y leaves no s: it is None, and the gradient, which needs the s, is not
    to be had."""
    dev, xt, wt, shape, dim, rp = _norm_args(x, weight, residual)
    out = _out(out, shape, x.dtype, x, "out")
    if rp is not None:
        total = _out(total, shape, x.dtype, x, "total")
    elif total is not None:
        raise ValueError("total needs a residual to add")
    rstd = torch.empty(shape[:-1], dtype=torch.float32, device=x.device)
    _call("muon_rms_norm", dev, x.data_ptr(), xt, rp, weight.data_ptr(), wt, rstd.numel(), dim, eps,
          None if rp is None else total.data_ptr(), out.data_ptr(), rstd.data_ptr())
    if rp is None:
        total = None if out.data_ptr() == x.data_ptr() and x.numel() else x
    return out, total, rstd


def muon_rms_norm8(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None, eps: float = 1e-6,
                   total: torch.Tensor | None = None):
    """muon_rms_norm with y in 8 bits: (y, scales, s, rstd), y float8_e4m3fn and
    scales fp32 [..., dim / 128 rounded up], a scale for each 128 columns."""
    dev, xt, wt, shape, dim, rp = _norm_args(x, weight, residual)
    y = torch.empty(shape, dtype=torch.float8_e4m3fn, device=x.device)
    scales = torch.empty((*shape[:-1], _blocks(dim)), dtype=torch.float32, device=x.device)
    if rp is not None:
        total = _out(total, shape, x.dtype, x, "total")
    elif total is not None:
        raise ValueError("total needs a residual to add")
    rstd = torch.empty(shape[:-1], dtype=torch.float32, device=x.device)
    _call("muon_rms_norm8", dev, x.data_ptr(), xt, rp, weight.data_ptr(), wt, rstd.numel(), dim, eps,
          None if rp is None else total.data_ptr(), y.data_ptr(), scales.data_ptr(), rstd.data_ptr())
    return y, scales, x if rp is None else total, rstd


def rms_norm_grad_workspace_size(rows: int, dim: int) -> int:
    return _size("muon_rms_norm_grad_workspace_size", int(rows), _int(int(dim), "dim"))


def muon_rms_norm_grad(dy: torch.Tensor, s: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor,
                       dsum: torch.Tensor | None = None, ds: torch.Tensor | None = None,
                       workspace: torch.Tensor | None = None):
    """Gradients of muon_rms_norm from the s and rstd it returned: (ds, dweight),
    ds (of x and of the residual) of s's dtype, dweight fp32.  `dsum`: the
    gradient that reaches s past the norm, added to ds.  `ds` may be dy, s or
    dsum.  Deterministic."""
    dev, xt, wt, shape, dim, _ = _norm_args(s, weight, None)
    for t, name in ((dy, "dy"), (dsum, "dsum"), (ds, "ds")):
        if t is not None or name == "dy":
            if _tensor(t, name, device=dev) != xt:
                raise TypeError(f"{name} must have s's dtype")
            _shaped(t, shape, name)
    _tensor(rstd, "rstd", _F32, dev)
    _shaped(rstd, shape[:-1], "rstd")
    if ds is None:
        ds = torch.empty_like(s)
    rows = rstd.numel()
    dweight = torch.empty((dim,), dtype=torch.float32, device=s.device)
    wp, wb, _keep = _workspace(workspace, dev, "muon_rms_norm_grad_workspace_size", rows, dim)
    _call("muon_rms_norm_grad", dev, dy.data_ptr(), s.data_ptr(), xt, weight.data_ptr(), wt, rstd.data_ptr(),
          None if dsum is None else dsum.data_ptr(), rows, dim, ds.data_ptr(), dweight.data_ptr(), wp, wb)
    return ds, dweight


def muon_quantize8(x: torch.Tensor, square: bool = False):
    """x in 8-bit storage: (q, scales), q float8_e4m3fn of x's shape, scales fp32:
    one for each 128 columns of a row ([..., dim / 128]), or with `square` for each
    128 x 128 block of the matrices of the last two axes ([..., rows / 128,
    dim / 128], rounded up), as muon_experts8 takes its W."""
    xt = _tensor(x, "x")
    shape = x.shape
    if len(shape) < (2 if square else 1):
        raise ValueError(f"x must have {'two axes' if square else 'an axis'}")
    dim = _int(shape[-1], "dim")
    rows = shape[-2] if square else (x.numel() // dim if dim else 0)
    batch = (x.numel() // (rows * dim) if rows and dim else 0) if square else 1
    lead = (*shape[:-2], _blocks(shape[-2])) if square else shape[:-1]
    q = torch.empty(shape, dtype=torch.float8_e4m3fn, device=x.device)
    scales = torch.empty((*lead, _blocks(dim)), dtype=torch.float32, device=x.device)
    _call("muon_quantize8", x.get_device(), x.data_ptr(), xt, batch, rows, dim, int(bool(square)), q.data_ptr(),
          scales.data_ptr())
    return q, scales


# ------------------------------------------------------------------ router --

def route_workspace_size(tokens: int, experts: int, k: int) -> int:
    return _size("muon_route_workspace_size", int(tokens), _int(int(experts), "experts"), _int(int(k), "k"))


def muon_route(logits: torch.Tensor, k: int, renormalize: bool = True, workspace: torch.Tensor | None = None):
    """The k experts of largest logit for each token and the plan that sorts the
    choices by expert: (gates, experts, slots, tokens, offsets).  logits
    [tokens][experts], bfloat16 or float32.  gates fp32 [tokens][k]: softmax at
    the choices, over all experts or (renormalize) over the choices; experts int32
    [tokens][k], -1 where fewer than k have a logit above -inf; slots int32
    [tokens][k], the row of each choice; tokens int32 [tokens * k], each row's
    token, -1 behind the last; offsets int32 [experts + 1], as muon_experts takes
    them.  muon_embed(x, tokens) brings rows to the experts, muon_combine brings
    theirs back."""
    t = _tensor(logits, "logits")
    dev = logits.get_device()
    if logits.dim() != 2:
        raise ValueError(f"logits must be [tokens][experts], got shape {tuple(logits.shape)}")
    n, e = logits.shape
    _int(e, "experts")
    _int(k, "k")
    wp, wb, _keep = _workspace(workspace, dev, "muon_route_workspace_size", n, e, k)
    gates = torch.empty((n, k), dtype=torch.float32, device=logits.device)
    chosen = torch.empty((n, k), dtype=torch.int32, device=logits.device)
    slots = torch.empty_like(chosen)
    tokens = torch.empty((n * k,), dtype=torch.int32, device=logits.device)
    offsets = torch.empty((e + 1,), dtype=torch.int32, device=logits.device)
    _call("muon_route", dev, logits.data_ptr(), t, n, e, k, bool(renormalize), gates.data_ptr(), chosen.data_ptr(),
          slots.data_ptr(), tokens.data_ptr(), offsets.data_ptr(), wp, wb)
    return gates, chosen, slots, tokens, offsets


def muon_route_grad(dgates: torch.Tensor, logits: torch.Tensor, experts: torch.Tensor,
                    renormalize: bool = True) -> torch.Tensor:
    """Gradient of muon_route's logits (of their dtype) from that of its gates
    (fp32), with the experts that it chose."""
    t = _tensor(logits, "logits")
    dev = logits.get_device()
    _tensor(dgates, "dgates", _F32, dev)
    _tensor(experts, "experts", _I32, dev)
    if logits.dim() != 2 or experts.dim() != 2 or experts.shape[0] != logits.shape[0]:
        raise ValueError(f"logits and experts must be [tokens][experts] and [tokens][k], got {tuple(logits.shape)} and "
                         f"{tuple(experts.shape)}")
    _shaped(dgates, experts.shape, "dgates")
    n, e = logits.shape
    dlogits = torch.empty_like(logits)
    _call("muon_route_grad", dev, dgates.data_ptr(), logits.data_ptr(), t, experts.data_ptr(), n, _int(e, "experts"),
          _int(experts.shape[1], "k"), bool(renormalize), dlogits.data_ptr())
    return dlogits


# ------------------------------------------------------------- combination --

def _combine_args(y, slots, gates):
    t = _tensor(y, "y")
    dev = y.get_device()
    _tensor(slots, "slots", _I32, dev)
    if y.dim() != 2 or slots.dim() != 2:
        raise ValueError(f"y and slots must be [rows][dim] and [tokens][k], got {tuple(y.shape)} and {tuple(slots.shape)}")
    gp = None
    if gates is not None:
        _tensor(gates, "gates", _F32, dev)
        _shaped(gates, slots.shape, "gates")
        gp = gates.data_ptr()
    return dev, t, gp, slots.shape[0], _int(slots.shape[1], "k"), y.shape[0], _int(y.shape[1], "dim")


def muon_combine(y: torch.Tensor, slots: torch.Tensor, gates: torch.Tensor | None = None,
                 out: torch.Tensor | None = None) -> torch.Tensor:
    """out[t] = the sum over j of gates[t][j] y[slots[t][j]], in fp32 and rounded
    once: y [rows][dim] bfloat16 or float32, slots int32 [tokens][k] (one outside
    the rows, such as -1, is left out), gates fp32 (1 without).  Without gates it
    is also the gradient of the dispatch muon_embed(x, tokens)."""
    dev, t, gp, n, k, rows, dim = _combine_args(y, slots, gates)
    out = _out(out, (n, dim), y.dtype, y, "out")
    _call("muon_combine", dev, y.data_ptr(), t, slots.data_ptr(), gp, n, k, rows, dim, out.data_ptr())
    return out


def muon_combine_grad(dout: torch.Tensor, y: torch.Tensor, slots: torch.Tensor, gates: torch.Tensor | None = None,
                      dy: torch.Tensor | None = None):
    """Gradients of muon_combine: (dy, dgates), dy of y's dtype, dgates fp32 (None
    without gates).  Each row is named by one slot at most, as muon_route does;
    rows that no slot names are not written (pass a zeroed `dy` if they are
    read)."""
    dev, t, gp, n, k, rows, dim = _combine_args(y, slots, gates)
    if _tensor(dout, "dout", device=dev) != t:
        raise TypeError("dout must have y's dtype")
    _shaped(dout, (n, dim), "dout")
    dy = _out(dy, (rows, dim), y.dtype, y, "dy")
    dgates = None if gates is None else torch.empty_like(gates)
    _call("muon_combine_grad", dev, dout.data_ptr(), y.data_ptr(), t, slots.data_ptr(), gp, n, k, rows, dim, dy.data_ptr(),
          None if dgates is None else dgates.data_ptr())
    return dy, dgates


# ----------------------------------------------------------------- experts --

def _experts_args(rows, rows_name, W, offsets, types, inner):
    """(device, rows, experts, out_dim, dim) of a grouped product whose rows
    have `inner` (1: out_dim, 2: dim) as their last axis."""
    _tensor(rows, rows_name, types)
    dev = rows.get_device()
    _tensor(W, "W", types, dev)
    _tensor(offsets, "offsets", _I32, dev)
    if rows.dim() != 2 or W.dim() != 3 or rows.shape[1] != W.shape[inner]:
        raise ValueError(f"{rows_name} and W must be [rows][{'out' if inner == 1 else 'dim'}] and [experts][out][dim], got "
                         f"{tuple(rows.shape)} and {tuple(W.shape)}")
    e, o, d = W.shape
    _shaped(offsets, (e + 1,), "offsets")
    return dev, rows.shape[0], _int(e, "experts"), _int(o, "out_dim"), _int(d, "dim")


def muon_experts(x: torch.Tensor, W: torch.Tensor, offsets: torch.Tensor, out: torch.Tensor | None = None,
                 error: torch.Tensor | None = None) -> torch.Tensor:
    """y[r] = W[e] x[r] for the rows offsets[e] <= r < offsets[e + 1] of each
    expert e: x bfloat16 [rows][dim], W bfloat16 [experts][out][dim], offsets
    int32 [experts + 1].  Rows of no expert are not written.  out and dim are
    multiples of 8.  What a wait on the device that ran out left uncomputed is
    NaN, and `error` (int32, optional) has the reason."""
    dev, n, e, o, d = _experts_args(x, "x", W, offsets, _BF16, 2)
    out = _out(out, (n, o), torch.bfloat16, x, "out")
    _call("muon_experts", dev, x.data_ptr(), W.data_ptr(), offsets.data_ptr(), n, e, o, d, out.data_ptr(), _error(error, dev))
    return out


def muon_experts_grad(dy: torch.Tensor, x: torch.Tensor | None, W: torch.Tensor, offsets: torch.Tensor,
                      dx: torch.Tensor | None = None, dW: torch.Tensor | None = None, accumulate: bool = False,
                      need_dx: bool = True, need_dW: bool = True, error: torch.Tensor | None = None):
    """Gradients of muon_experts: (dx, dW), dx bfloat16 (rows of no expert not
    written), dW float32 unless a bfloat16 `dW` is given, zero for an expert
    without rows; with `accumulate` it is added to a float32 dW.  need_dx or
    need_dW False: that one is not computed, and None; x is read for dW alone and may
    be None without it."""
    dev, n, e, o, d = _experts_args(dy, "dy", W, offsets, _BF16, 1)
    if x is not None or need_dW:
        _tensor(x, "x", _BF16, dev)
        _shaped(x, (n, d), "x")
    dx = _out(dx, (n, d), torch.bfloat16, dy, "dx") if need_dx else None
    wt = 1
    if not need_dW:
        dW = None
    elif dW is None:
        if accumulate:
            raise ValueError("accumulate needs the dW to add to")
        dW = torch.empty((e, o, d), dtype=torch.float32, device=dy.device)
    else:
        wt = _tensor(dW, "dW", device=dev)
        _shaped(dW, (e, o, d), "dW")
    _call("muon_experts_grad", dev, dy.data_ptr(), None if x is None else x.data_ptr(), W.data_ptr(), offsets.data_ptr(), n, e, o, d,
          None if dx is None else dx.data_ptr(), None if dW is None else dW.data_ptr(), wt, bool(accumulate),
          _error(error, dev))
    return dx, dW


def muon_experts8(x: torch.Tensor, x_scales: torch.Tensor, W: torch.Tensor, W_scales: torch.Tensor,
                  offsets: torch.Tensor, out: torch.Tensor | None = None, error: torch.Tensor | None = None) -> torch.Tensor:
    """muon_experts of 8-bit operands (float8_e4m3fn values with float32 scales):
    x_scales [rows][dim / 128], W_scales [experts][out / 128][dim / 128], both
    rounded up, as muon_rms_norm8 and muon_quantize8 write them.  y is bfloat16;
    dim is a multiple of 16, out of 8."""
    dev, n, e, o, d = _experts_args(x, "x", W, offsets, _E4M3, 2)
    _tensor(x_scales, "x_scales", _F32, dev)
    _tensor(W_scales, "W_scales", _F32, dev)
    _shaped(x_scales, (n, _blocks(d)), "x_scales")
    _shaped(W_scales, (e, _blocks(o), _blocks(d)), "W_scales")
    out = _out(out, (n, o), torch.bfloat16, x, "out")
    _call("muon_experts8", dev, x.data_ptr(), x_scales.data_ptr(), W.data_ptr(), W_scales.data_ptr(), offsets.data_ptr(), n,
          e, o, d, out.data_ptr(), _error(error, dev))
    return out
