"""The global gradient norm over many tensors, and clipping.

    norm = clip_grad_norm_(grads, 1.0)                      # in place, as a training loop does
    norm = clip_grad_norm_([out["dW"], *rest], 1.0,         # the head's fp32 gradient and the
                           out=[W_grad_bf16, *rest_grads])  # others, clipped into other tensors

Everything is enqueued on the current stream of the tensors' device, and the norm
stays on the device: no synchronisation."""
from __future__ import annotations

import array
import math

import torch

from . import _lib as L
from .ops import on_device

_DT = {torch.bfloat16: L.KL_DTYPE_BF16, torch.float32: L.KL_DTYPE_F32,
       torch.float16: L.KL_DTYPE_F16}


def _dense(t):
    """Whether t's elements fill one block of memory, each once, in some order."""
    order = sorted(range(t.dim()), key=t.stride, reverse=True)
    return t.permute(order).is_contiguous()


def _list(ts, name):
    """The tensors as a list, their device, and the library's names of their types."""
    ts = [ts] if isinstance(ts, torch.Tensor) else list(ts)
    if not ts:
        raise ValueError(f"no {name}")
    try:
        where = set(map(torch.Tensor.get_device, ts))
    except TypeError:
        raise ValueError(f"{name} must be tensors") from None
    if len(where) != 1 or where == {-1}:
        raise ValueError(f"{name} must be on one CUDA device")
    try:
        return ts, ts[0].device, [_DT[t.dtype] for t in ts]
    except KeyError:
        raise TypeError(f"{name} must be float32, bfloat16 or float16") from None


def _table(src, dst=None):
    """The library's table of the tensors (an array that stays alive for the call),
    their number and device."""
    src, dev, st = _list(src, "gradients")
    if dst is None:
        if not all(map(torch.Tensor.is_contiguous, src)) and not all(
                t.is_contiguous() or _dense(t) for t in src):
            raise ValueError("a gradient with gaps or repeats in memory")
        to = at = list(map(torch.Tensor.data_ptr, src))
        dt = st
    else:
        dst, dev_d, dt = _list(dst, "destinations")
        if len(src) != len(dst) or dev_d != dev:
            raise ValueError(f"{len(src)} gradients on {dev}, {len(dst)} destinations on {dev_d}")
        for s, d in zip(src, dst):
            if s.shape != d.shape or not s.is_contiguous() or not d.is_contiguous():
                raise ValueError("a destination must be contiguous, of its gradient's shape")
        at, to = (list(map(torch.Tensor.data_ptr, ts)) for ts in (src, dst))
    # kl_grad: src, dst, n, and the two 32-bit types in one word
    kinds = [a | b << 32 for a, b in zip(st, dt)]
    table = array.array("q", bytes(32 * len(src)))
    for column, values in enumerate((at, to, map(torch.Tensor.numel, src), kinds)):
        table[column::4] = array.array("q", values)
    return table, len(src), dev


_requires_grad = torch.Tensor.requires_grad.__get__


def _no_parameters(ts):
    """Refuses parameters, whose weights would be scaled (or overwritten) in place of
    their gradients."""
    if any(map(_requires_grad, ts)) and any(t.requires_grad and t.is_leaf for t in ts):
        raise ValueError("a leaf that requires grad: pass its gradient (p.grad), not the "
                         "parameter")


def _norm_type(norm_type):
    if norm_type == 2:
        return L.KL_NORM_2
    if norm_type in (math.inf, "inf"):
        return L.KL_NORM_INF
    raise ValueError("norm_type must be 2 or inf")


def _scratch(n, dev):
    return torch.empty(L.kl_grad_workspace_bytes(n), dtype=torch.uint8, device=dev)


def _norm(grads, norm_type, dtype):
    table, n, dev = _table(grads)
    kind, ws = _norm_type(norm_type), _scratch(n, dev)
    out = torch.empty((), dtype=dtype, device=dev)
    total, norm = (out.data_ptr(), None) if dtype == torch.float64 else (None, out.data_ptr())
    on_device(dev, "kl_grad_norm", table.buffer_info()[0], n, kind, ws.data_ptr(), ws.numel(),
              total, norm)
    return out


def grad_norm(grads, *, norm_type=2.0):
    """Norm of all values of the tensors (float32 device scalar): the root of the sum
    of squares, or with norm_type inf the largest magnitude.  Squares beyond float32's
    range count too."""
    return _norm(grads, norm_type, torch.float32)


def grad_total(grads, *, norm_type=2.0):
    """The sum of squares (norm_type 2) or the largest magnitude as a float64 device
    scalar: what ranks that hold parts of the gradients join, for clip_grad_norm_."""
    return _norm(grads, norm_type, torch.float64)


def clip_grad_norm_(grads, max_norm, *, norm_type=2.0, out=None, total=None):
    """Scales the gradients by min(1, max_norm / (norm + 1e-6)) and returns the norm
    before (float32 device scalar).  grads are the gradients themselves, not the
    parameters: a leaf that requires grad is refused.  In place, or into the tensors
    `out`, each rounded once to its type.  In place nothing is written while the norm
    stays under max_norm.  total: the float64 device scalar that grad_total gives (joined
    over ranks, say) in place of the tensors' own.  A NaN norm gives NaN everywhere, an
    infinite one zeros (NaN where a gradient is infinite)."""
    grads, out = ([ts] if isinstance(ts, torch.Tensor) else ts if ts is None else list(ts)
                  for ts in (grads, out))
    table, n, dev = _table(grads, out)
    _no_parameters(grads if out is None else grads + out)
    kind, ws = _norm_type(norm_type), _scratch(n, dev)
    if total is not None and (not isinstance(total, torch.Tensor) or total.numel() != 1 or
                              total.dtype != torch.float64 or total.device != dev):
        raise ValueError("total must be a float64 scalar on the gradients' device")
    norm = torch.empty((), dtype=torch.float32, device=dev)
    on_device(dev, "kl_grad_clip", table.buffer_info()[0], n, kind, float(max_norm),
              None if total is None else total.data_ptr(), ws.data_ptr(), ws.numel(),
              norm.data_ptr())
    return norm
