"""Binding of include/muon_lm.h: the operators at the ends of a language model.

As in ns.py, argument marshalling only; names follow the C entry points.
Tensors are contiguous CUDA tensors of bfloat16 or float32 on one device, and
work is enqueued on that device's current stream.  The head's h and table are
bfloat16, with a dim that is a multiple of 8.  As everywhere in this package,
autograd is not involved: results require no gradient whatever the arguments
do, and the backward pass is the caller's to call.  The small calls take about
as long to issue as to run, so the checks here are kept to a few tests a
tensor.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import _lib

_BF16 = {torch.bfloat16: 0}
_F32 = {torch.float32: 1}
_TYPES = {torch.bfloat16: 0, torch.float32: 1}
_IDS = {torch.int32: 32, torch.int64: 64}


def _tensor(t, name, types=_TYPES, device=None):
    """The C type code of a contiguous CUDA tensor of one of `types` (and on
    CUDA device number `device`)."""
    code = types.get(t.dtype) if isinstance(t, torch.Tensor) else None
    if code is None or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor of {', '.join(str(k) for k in types)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if device is not None and t.get_device() != device:
        raise ValueError(f"{name} must be on cuda:{device}")
    return code


def _shaped(t, shape, name):
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _int(n, name):
    """n, refused if it does not fit a C int: ctypes would keep its low bits."""
    if not -1 << 31 <= n < 1 << 31:
        raise _lib.MuonNSError(_lib.ERR_INVALID_ARG, f"{name} {n}")
    return n


# The current stream's handle without a Stream object around it, where this
# PyTorch has it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)


@functools.lru_cache(maxsize=None)
def _entry(name):
    return getattr(_lib.lib(), name)


def _call(name, device, *args):
    """Calls a C entry point on CUDA device number `device`, its current stream
    last."""
    if torch.cuda.current_device() == device:
        s = _entry(name)(*args, _raw_stream(device))
    else:
        with torch.cuda.device(device):
            s = _entry(name)(*args, _raw_stream(device))
    if s != _lib.OK:
        _lib.check(s, name)


@functools.lru_cache(maxsize=1024)
def _size(name, *args) -> int:
    """Workspace bytes: a function of the sizes alone."""
    n = ctypes.c_size_t(0)
    _lib.check(_entry(name)(*args, ctypes.byref(n)), name)
    return n.value


def _workspace(workspace, device, name, *args):
    """(pointer, bytes, tensor to keep) of the caller's workspace or a new one."""
    if workspace is None:
        n = _size(name, *args)
        if n == 0:
            return None, 0, None
        workspace = torch.empty(n, dtype=torch.uint8, device=device)
        return workspace.data_ptr(), n, workspace
    if not isinstance(workspace, torch.Tensor) or not workspace.is_contiguous() or workspace.get_device() != device:
        raise ValueError(f"workspace must be a contiguous tensor on cuda:{device}")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


# --------------------------------------------------------------- embedding --

def muon_embed(table: torch.Tensor, ids: torch.Tensor, scale: float = 1.0, dtype: torch.dtype | None = None,
               out: torch.Tensor | None = None) -> torch.Tensor:
    """out[t] = scale * table[ids[t]] for int32 or int64 ids of any shape;
    rows of ids outside [0, vocab) are zero.  `dtype`: of the result (the
    table's)."""
    tt = _tensor(table, "table")
    dev = table.get_device()
    ib = _tensor(ids, "ids", _IDS, dev)
    if table.dim() != 2:
        raise ValueError(f"table must be [vocab][dim], got shape {tuple(table.shape)}")
    vocab, dim = table.shape
    _int(dim, "dim")
    shape = (*ids.shape, dim)
    if out is None:
        out = torch.empty(shape, dtype=dtype or table.dtype, device=table.device)
        ot = _TYPES.get(out.dtype)
        if ot is None:
            raise TypeError(f"dtype must be one of {', '.join(str(k) for k in _TYPES)}")
    else:
        ot = _tensor(out, "out", device=dev)
        _shaped(out, shape, "out")
        if dtype is not None and out.dtype != dtype:
            raise ValueError("out must have the dtype asked for")
    _call("muon_embed", dev, table.data_ptr(), tt, vocab, dim, ids.data_ptr(), ib, ids.numel(), scale, out.data_ptr(), ot)
    return out


def embed_grad_workspace_size(tokens: int, vocab: int, dim: int) -> int:
    return _size("muon_embed_grad_workspace_size", int(tokens), int(vocab), _int(int(dim), "dim"))


def muon_embed_grad(dy: torch.Tensor, ids: torch.Tensor, vocab: int, scale: float = 1.0,
                    dtable: torch.Tensor | None = None, accumulate: bool = False,
                    workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Gradient of muon_embed's table: dtable[v] = scale * the sum of dy over
    the tokens with id v (fp32 [vocab][dim] unless `dtable` is given; with
    `accumulate` it is added to dtable).  Deterministic."""
    dt = _tensor(dy, "dy")
    dev = dy.get_device()
    ib = _tensor(ids, "ids", _IDS, dev)
    if dy.dim() != ids.dim() + 1:
        raise ValueError("dy must have one more axis than ids")
    dim = _int(dy.shape[-1], "dim")
    _shaped(dy, (*ids.shape, dim), "dy")
    if dtable is None:
        if accumulate:
            raise ValueError("accumulate needs the dtable to add to")
        dtable = torch.empty((vocab, dim), dtype=torch.float32, device=dy.device)
        ot = 1
    else:
        ot = _tensor(dtable, "dtable", device=dev)
        _shaped(dtable, (vocab, dim), "dtable")
    n = ids.numel()
    wp, wb, _keep = _workspace(workspace, dev, "muon_embed_grad_workspace_size", n, vocab, dim)
    _call("muon_embed_grad", dev, dy.data_ptr(), dt, ids.data_ptr(), ib, n, vocab, dim, scale, dtable.data_ptr(), ot,
          bool(accumulate), wp, wb)
    return dtable


# -------------------------------------------------------------- layer norm --

def muon_layer_norm(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None = None, eps: float = 1e-5,
                    out: torch.Tensor | None = None):
    """Layer norm over the last axis.  Returns (y, mean, rstd): y of x's shape
    and dtype, mean and rstd fp32 of x's shape without its last axis.  weight
    and bias: bfloat16 or float32, one dtype.  `out` may be x."""
    xt = _tensor(x, "x")
    dev = x.get_device()
    wt = _tensor(weight, "weight", device=dev)
    shape = x.shape
    if not shape:
        raise ValueError("x must have an axis to normalise over")
    dim = _int(shape[-1], "dim")
    _shaped(weight, (dim,), "weight")
    bp = None
    if bias is not None:
        if _tensor(bias, "bias", device=dev) != wt:
            raise TypeError("bias must have weight's dtype")
        _shaped(bias, (dim,), "bias")
        bp = bias.data_ptr()
    if out is None:
        out = torch.empty_like(x)
    else:
        if _tensor(out, "out", device=dev) != xt:
            raise TypeError("out must have x's dtype")
        _shaped(out, shape, "out")
    mean = torch.empty(shape[:-1], dtype=torch.float32, device=x.device)
    rstd = torch.empty_like(mean)
    _call("muon_layer_norm", dev, x.data_ptr(), xt, weight.data_ptr(), bp, wt, mean.numel(), dim, eps, out.data_ptr(),
          mean.data_ptr(), rstd.data_ptr())
    return out, mean, rstd


def layer_norm_grad_workspace_size(rows: int, dim: int) -> int:
    return _size("muon_layer_norm_grad_workspace_size", int(rows), _int(int(dim), "dim"))


def muon_layer_norm_grad(dy: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, mean: torch.Tensor,
                         rstd: torch.Tensor, bias: bool = True, dx: torch.Tensor | None = None,
                         workspace: torch.Tensor | None = None):
    """Gradients of muon_layer_norm from the mean and rstd it returned: (dx,
    dweight, dbias), dx of x's dtype, dweight and dbias fp32 (dbias None with
    bias=False).  `dx` may be dy or x.  Deterministic."""
    xt = _tensor(x, "x")
    dev = x.get_device()
    if _tensor(dy, "dy", device=dev) != xt:
        raise TypeError("dy must have x's dtype")
    wt = _tensor(weight, "weight", device=dev)
    shape = x.shape
    if not shape:
        raise ValueError("x must have an axis to normalise over")
    dim, lead = _int(shape[-1], "dim"), shape[:-1]
    _shaped(dy, shape, "dy")
    _shaped(weight, (dim,), "weight")
    _tensor(mean, "mean", _F32, dev)
    _tensor(rstd, "rstd", _F32, dev)
    _shaped(mean, lead, "mean")
    _shaped(rstd, lead, "rstd")
    if dx is None:
        dx = torch.empty_like(x)
    else:
        if _tensor(dx, "dx", device=dev) != xt:
            raise TypeError("dx must have x's dtype")
        _shaped(dx, shape, "dx")
    rows = mean.numel()
    dweight = torch.empty((dim,), dtype=torch.float32, device=x.device)
    dbias = torch.empty_like(dweight) if bias else None
    wp, wb, _keep = _workspace(workspace, dev, "muon_layer_norm_grad_workspace_size", rows, dim)
    _call("muon_layer_norm_grad", dev, dy.data_ptr(), x.data_ptr(), xt, weight.data_ptr(), wt, mean.data_ptr(),
          rstd.data_ptr(), rows, dim, dx.data_ptr(), dweight.data_ptr(), dbias.data_ptr() if bias else None, wp, wb)
    return dx, dweight, dbias


# -------------------------------------------------------------------- head --

def head_workspace_size(tokens: int, vocab: int, dim: int, grad: bool = True, pieces: int = 0) -> int:
    return _size("muon_head_workspace_size", int(tokens), int(vocab), _int(int(dim), "dim"), int(bool(grad)),
                 _int(int(pieces), "pieces"))


def _head_args(h, table, targets):
    _tensor(h, "h", _BF16)
    dev = h.get_device()
    _tensor(table, "table", _BF16, dev)
    bits = _tensor(targets, "targets", _IDS, dev)
    shape = h.shape
    if not shape or table.dim() != 2 or table.shape[1] != shape[-1]:
        raise ValueError(f"h and table must be [...][dim] and [vocab][dim], got {tuple(shape)} and {tuple(table.shape)}")
    _shaped(targets, shape[:-1], "targets")
    return dev, bits, targets.numel(), table.shape[0], _int(table.shape[1], "dim")


def muon_head_loss(h: torch.Tensor, table: torch.Tensor, targets: torch.Tensor, ignore_index: int = -100,
                   workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Cross entropy of softmax(h table^T) at `targets`, a loss a token (fp32
    of targets' shape), without logits in memory.  h and table are bfloat16;
    targets int32 or int64.  Tokens whose target is ignore_index or outside
    the table have loss 0.  If a wait on the device runs out
    (set_wait_budget), every loss is NaN; a `workspace` of the caller's has the
    reason (read_error, muon_ns_check)."""
    dev, bits, n, vocab, dim = _head_args(h, table, targets)
    loss = torch.empty(targets.shape, dtype=torch.float32, device=h.device)
    wp, wb, _keep = _workspace(workspace, dev, "muon_head_workspace_size", n, vocab, dim, 0, 0)
    _call("muon_head_loss", dev, h.data_ptr(), table.data_ptr(), n, vocab, dim, targets.data_ptr(), bits, ignore_index,
          loss.data_ptr(), wp, wb)
    return loss


def muon_head_loss_grad(h: torch.Tensor, table: torch.Tensor, targets: torch.Tensor, ignore_index: int = -100,
                        dloss: torch.Tensor | None = None, dtable: torch.Tensor | None = None,
                        accumulate: bool = False, pieces: int = 0, workspace: torch.Tensor | None = None):
    """(loss, dh, dtable): muon_head_loss and the gradient of sum(dloss * loss)
    in one call; dloss (fp32 of targets' shape) defaults to the mean's, 1 / the
    number of tokens with a loss.  dh is bfloat16; dtable bfloat16 unless a
    float32 `dtable` is given, to which `accumulate` adds (its products' operands
    are bfloat16 all the same).  The workspace holds the bfloat16 probabilities
    of one of `pieces` of the vocabulary (0: pieces of about 4 GiB; more than
    one cost up to a third more work).  If a wait on the
    device runs out, all three are NaN throughout, as in muon_head_loss."""
    dev, bits, n, vocab, dim = _head_args(h, table, targets)
    _int(pieces, "pieces")
    dp = None
    if dloss is not None:
        _tensor(dloss, "dloss", _F32, dev)
        _shaped(dloss, targets.shape, "dloss")
        dp = dloss.data_ptr()
    if dtable is None:
        if accumulate:
            raise ValueError("accumulate needs the dtable to add to")
        dtable = torch.empty_like(table)
        dt = 0
    else:
        dt = _tensor(dtable, "dtable", device=dev)
        _shaped(dtable, table.shape, "dtable")
    loss = torch.empty(targets.shape, dtype=torch.float32, device=h.device)
    dh = torch.empty_like(h)
    wp, wb, _keep = _workspace(workspace, dev, "muon_head_workspace_size", n, vocab, dim, 1, pieces)
    _call("muon_head_loss_grad", dev, h.data_ptr(), table.data_ptr(), n, vocab, dim, targets.data_ptr(), bits,
          ignore_index, dp, pieces, loss.data_ptr(), dh.data_ptr(), dtable.data_ptr(), dt, bool(accumulate), wp, wb)
    return loss, dh, dtable
