"""Binding of include/muon_lm.h: the operators at the ends of a language model.

As in ns.py, argument marshalling only; names follow the C entry points.
Tensors are contiguous CUDA tensors of bfloat16 or float32 on one device, and
work is enqueued on that device's current stream.
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib

_TYPES = {torch.bfloat16: 0, torch.float32: 1}
_IDS = {torch.int32: 32, torch.int64: 64}


def _tensor(t, name, types=_TYPES, device=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype not in types:
        raise TypeError(f"{name} must be a CUDA tensor of {', '.join(str(k) for k in types)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}")
    return types[t.dtype]


_F32 = {torch.float32: 1}


def _shaped(t, shape, name):
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _call(name, device, *args):
    """Calls the C entry point with the current stream of `device` last."""
    fn = getattr(_lib.lib(), name)
    if torch.cuda.current_device() == device.index:
        s = fn(*args, torch.cuda.current_stream(device).cuda_stream)
    else:
        with torch.cuda.device(device):
            s = fn(*args, torch.cuda.current_stream(device).cuda_stream)
    if s != _lib.OK:
        _lib.check(s, name)


def _size(name, *args) -> int:
    n = ctypes.c_size_t(0)
    _lib.check(getattr(_lib.lib(), name)(*args, ctypes.byref(n)), name)
    return n.value


def _workspace(workspace, bytes_, device):
    if workspace is None:
        return torch.empty(max(bytes_, 1), dtype=torch.uint8, device=device)
    if not isinstance(workspace, torch.Tensor) or not workspace.is_contiguous() or workspace.device != device:
        raise ValueError(f"workspace must be a contiguous tensor on {device}")
    return workspace


def _nbytes(t):
    return t.numel() * t.element_size()


# --------------------------------------------------------------- embedding --

def muon_embed(table: torch.Tensor, ids: torch.Tensor, scale: float = 1.0, dtype: torch.dtype | None = None,
               out: torch.Tensor | None = None) -> torch.Tensor:
    """out[t] = scale * table[ids[t]] for int32 or int64 ids of any shape;
    rows of ids outside [0, vocab) are zero.  `dtype`: of the result (the
    table's)."""
    tt = _tensor(table, "table")
    ib = _tensor(ids, "ids", _IDS, table.device)
    if table.dim() != 2:
        raise ValueError(f"table must be [vocab][dim], got shape {tuple(table.shape)}")
    vocab, dim = table.shape
    if out is None:
        out = torch.empty((*ids.shape, dim), dtype=dtype or table.dtype, device=table.device)
    ot = _tensor(out, "out", device=table.device)
    _shaped(out, (*ids.shape, dim), "out")
    if dtype is not None and out.dtype != dtype:
        raise ValueError("out must have the dtype asked for")
    _call("muon_embed", table.device, table.data_ptr(), tt, vocab, dim, ids.data_ptr(), ib, ids.numel(), float(scale),
          out.data_ptr(), ot)
    return out


def embed_grad_workspace_size(tokens: int, vocab: int, dim: int) -> int:
    return _size("muon_embed_grad_workspace_size", int(tokens), int(vocab), int(dim))


def muon_embed_grad(dy: torch.Tensor, ids: torch.Tensor, vocab: int, scale: float = 1.0,
                    dtable: torch.Tensor | None = None, accumulate: bool = False,
                    workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Gradient of muon_embed's table: dtable[v] = scale * the sum of dy over
    the tokens with id v (fp32 [vocab][dim] unless `dtable` is given; with
    `accumulate` it is added to dtable).  Deterministic."""
    dt = _tensor(dy, "dy")
    ib = _tensor(ids, "ids", _IDS, dy.device)
    if dy.dim() != ids.dim() + 1:
        raise ValueError("dy must have one more axis than ids")
    dim = dy.shape[-1]
    _shaped(dy, (*ids.shape, dim), "dy")
    if dtable is None:
        if accumulate:
            raise ValueError("accumulate needs the dtable to add to")
        dtable = torch.empty((vocab, dim), dtype=torch.float32, device=dy.device)
    ot = _tensor(dtable, "dtable", device=dy.device)
    _shaped(dtable, (vocab, dim), "dtable")
    n = ids.numel()
    if workspace is None:
        workspace = _workspace(None, embed_grad_workspace_size(n, vocab, dim), dy.device)
    else:
        _workspace(workspace, 0, dy.device)
    _call("muon_embed_grad", dy.device, dy.data_ptr(), dt, ids.data_ptr(), ib, n, vocab, dim, float(scale),
          dtable.data_ptr(), ot, int(bool(accumulate)), workspace.data_ptr(), _nbytes(workspace))
    return dtable


# -------------------------------------------------------------- layer norm --

def muon_layer_norm(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None = None, eps: float = 1e-5,
                    out: torch.Tensor | None = None):
    """Layer norm over the last axis.  Returns (y, mean, rstd): y of x's shape
    and dtype, mean and rstd fp32 of x's shape without its last axis.  weight
    and bias: bfloat16 or float32, one dtype.  `out` may be x."""
    xt = _tensor(x, "x")
    wt = _tensor(weight, "weight", device=x.device)
    if x.dim() < 1:
        raise ValueError("x must have an axis to normalise over")
    dim = x.shape[-1]
    _shaped(weight, (dim,), "weight")
    if bias is not None:
        if _tensor(bias, "bias", device=x.device) != wt:
            raise TypeError("bias must have weight's dtype")
        _shaped(bias, (dim,), "bias")
    if out is None:
        out = torch.empty_like(x)
    if _tensor(out, "out", device=x.device) != xt:
        raise TypeError("out must have x's dtype")
    _shaped(out, x.shape, "out")
    stat = torch.empty((2, *x.shape[:-1]), dtype=torch.float32, device=x.device)
    mean, rstd = stat[0], stat[1]
    rows = mean.numel()
    _call("muon_layer_norm", x.device, x.data_ptr(), xt, weight.data_ptr(), None if bias is None else bias.data_ptr(),
          wt, rows, dim, float(eps), out.data_ptr(), mean.data_ptr(), rstd.data_ptr())
    return out, mean, rstd


def layer_norm_grad_workspace_size(rows: int, dim: int) -> int:
    return _size("muon_layer_norm_grad_workspace_size", int(rows), int(dim))


def muon_layer_norm_grad(dy: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, mean: torch.Tensor,
                         rstd: torch.Tensor, bias: bool = True, dx: torch.Tensor | None = None,
                         workspace: torch.Tensor | None = None):
    """Gradients of muon_layer_norm from the mean and rstd it returned: (dx,
    dweight, dbias), dx of x's dtype, dweight and dbias fp32 (dbias None with
    bias=False).  `dx` may be dy or x.  Deterministic."""
    xt = _tensor(x, "x")
    dev = x.device
    if _tensor(dy, "dy", device=dev) != xt:
        raise TypeError("dy must have x's dtype")
    wt = _tensor(weight, "weight", device=dev)
    if x.dim() < 1:
        raise ValueError("x must have an axis to normalise over")
    dim = x.shape[-1]
    _shaped(dy, x.shape, "dy")
    _shaped(weight, (dim,), "weight")
    for t, n in ((mean, "mean"), (rstd, "rstd")):
        _tensor(t, n, _F32, dev)
        _shaped(t, x.shape[:-1], n)
    if dx is None:
        dx = torch.empty_like(x)
    if _tensor(dx, "dx", device=dev) != xt:
        raise TypeError("dx must have x's dtype")
    _shaped(dx, x.shape, "dx")
    rows = mean.numel()
    grads = torch.empty((2 if bias else 1, dim), dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = _workspace(None, layer_norm_grad_workspace_size(rows, dim), dev)
    else:
        _workspace(workspace, 0, dev)
    dbias = grads[1] if bias else None
    _call("muon_layer_norm_grad", dev, dy.data_ptr(), x.data_ptr(), xt, weight.data_ptr(), wt, mean.data_ptr(),
          rstd.data_ptr(), rows, dim, dx.data_ptr(), grads.data_ptr(), dbias.data_ptr() if bias else None,
          workspace.data_ptr(), _nbytes(workspace))
    return dx, grads[0], dbias


# -------------------------------------------------------------------- head --

_BF16 = {torch.bfloat16: 0}


def head_workspace_size(tokens: int, vocab: int, dim: int, grad: bool = True, pieces: int = 0) -> int:
    return _size("muon_head_workspace_size", int(tokens), int(vocab), int(dim), int(bool(grad)), int(pieces))


def _head_args(h, table, targets):
    _tensor(h, "h", _BF16)
    dev = h.device
    _tensor(table, "table", _BF16, dev)
    bits = _tensor(targets, "targets", _IDS, dev)
    if h.dim() < 1 or table.dim() != 2 or table.shape[1] != h.shape[-1]:
        raise ValueError(f"h and table must be [...][dim] and [vocab][dim], got {tuple(h.shape)} and {tuple(table.shape)}")
    _shaped(targets, h.shape[:-1], "targets")
    return dev, bits, targets.numel(), table.shape[0], table.shape[1]


def muon_head_loss(h: torch.Tensor, table: torch.Tensor, targets: torch.Tensor, ignore_index: int = -100,
                   workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Cross entropy of softmax(h table^T) at `targets`, a loss a token (fp32
    of targets' shape), without keeping the logits.  h and table are bfloat16;
    targets int32 or int64.  Tokens whose target is ignore_index or outside
    the table have loss 0."""
    dev, bits, n, vocab, dim = _head_args(h, table, targets)
    loss = torch.empty(targets.shape, dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = _workspace(None, head_workspace_size(n, vocab, dim, False), dev)
    else:
        _workspace(workspace, 0, dev)
    _call("muon_head_loss", dev, h.data_ptr(), table.data_ptr(), n, vocab, dim, targets.data_ptr(), bits,
          int(ignore_index), loss.data_ptr(), workspace.data_ptr(), _nbytes(workspace))
    return loss


def muon_head_loss_grad(h: torch.Tensor, table: torch.Tensor, targets: torch.Tensor, ignore_index: int = -100,
                        dloss: torch.Tensor | None = None, dtable: torch.Tensor | None = None,
                        accumulate: bool = False, pieces: int = 0, workspace: torch.Tensor | None = None):
    """(loss, dh, dtable): muon_head_loss and the gradient of sum(dloss * loss)
    in one call; dloss (fp32 of targets' shape) defaults to the mean's, 1 / the
    number of tokens with a loss.  dh is bfloat16; dtable bfloat16 unless a
    float32 `dtable` is given, to which `accumulate` adds.  `pieces` of the
    vocabulary bound the workspace (0: pieces of about 4 GiB)."""
    dev, bits, n, vocab, dim = _head_args(h, table, targets)
    if dloss is not None:
        _tensor(dloss, "dloss", _F32, dev)
        _shaped(dloss, targets.shape, "dloss")
    if dtable is None:
        if accumulate:
            raise ValueError("accumulate needs the dtable to add to")
        dtable = torch.empty_like(table)
    dt = _tensor(dtable, "dtable", device=dev)
    _shaped(dtable, table.shape, "dtable")
    loss = torch.empty(targets.shape, dtype=torch.float32, device=dev)
    dh = torch.empty_like(h)
    if workspace is None:
        workspace = _workspace(None, head_workspace_size(n, vocab, dim, True, pieces), dev)
    else:
        _workspace(workspace, 0, dev)
    _call("muon_head_loss_grad", dev, h.data_ptr(), table.data_ptr(), n, vocab, dim, targets.data_ptr(), bits,
          int(ignore_index), None if dloss is None else dloss.data_ptr(), int(pieces), loss.data_ptr(), dh.data_ptr(),
          dtable.data_ptr(), dt, int(bool(accumulate)), workspace.data_ptr(), _nbytes(workspace))
    return loss, dh, dtable
